"""Products of 8-bit integers over rows grouped by expert: exact sums, so every
element is held to the four roundings behind them."""
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


def _codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int32).to(torch.int8)


def _scales(shape, seed, at=1.0):
    g = torch.Generator().manual_seed(seed)
    return (0.5 + torch.rand(shape, generator=g)) * at


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(cco, first, count, rows, n, k, dtype, seed=0, ld=None, sld=1, shift=0):
    """One product against exact sums; rows of no group and the columns behind
    the result stay as they were.  ld: row distance of x and y; sld: of xs;
    shift: elements the operands lie past an aligned address."""
    say("case: i8 product %s groups=%d rows=%d n=%d k=%d ld=%s shift=%d" % (
        dtype, len(first), rows, n, k, ld, shift))
    G = len(first)
    x, w = _codes((rows, k), seed + 1), _codes((G, n, k), seed + 2)
    # (results within fp16's range)
    xs, ws = _scales(rows, seed + 3, 1.0 / 128), _scales((G, n), seed + 4, 1.0 / (16 * k ** 0.5))
    ldx, ldy = ld or (k, n)

    def place(t, pitch, fill):
        flat = torch.full((shift + t.shape[0] * pitch,), fill, dtype=t.dtype, device="cuda")
        v = flat[shift:].view(t.shape[0], pitch)[:, :t.shape[1]]
        v.copy_(t)
        return v, flat

    xd, _ = place(x, ldx, 99)
    wd = torch.empty(shift + w.numel(), dtype=torch.int8, device="cuda")[shift:].view(w.shape)
    wd.copy_(w)
    xsd = torch.full((rows, sld), math.nan, device="cuda")
    xsd[:, 0] = xs
    y, flat = place(torch.full((rows, n), 7.0, dtype=dtype), ldy, 7.0)
    got = cco.group_product_i8(_i32(first), _i32(count), xd, xsd[:, 0], wd, ws.cuda(), out=y)
    assert got is y
    want = serve_ref.product_i8(first, count, x, xs, w, ws,
                                torch.full((rows, n), 7.0, dtype=torch.float64))
    ops_ref.assert_within(y, want, serve_ref.product_i8_bound(want, dtype), "y")
    if ldy > n:
        behind = flat[shift:].view(rows, ldy)[:, n:]
        assert bool((behind == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", [(1, 8, 16), (1, 1, 1), (3, 5, 7), (31, 24, 48), (33, 40, 15),
                                      (64, 129, 127), (130, 136, 144), (127, 300, 200),
                                      (257, 520, 1040), (300, 264, 4096), (1000, 256, 128)])
def test_one_group(cco, dtype, rows, n, k):
    _check(cco, [0], [rows], rows, n, k, dtype, rows + n)


@pytest.mark.parametrize("n,k", [(256, 512), (264, 528), (1000, 1416), (513, 2048), (40, 65)])
def test_ragged_groups(cco, n, k):
    count = [0, 1, 130, 0, 256, 31, 300, 2, 0]
    first = [sum(count[:i]) for i in range(len(count))]
    _check(cco, first, count, sum(count), n, k, torch.bfloat16, 3)


def test_groups_that_leave_rows_out_and_pass_the_ends(cco):
    # rows 0..4 and 20..29 belong to no group; counts below zero and past the end
    for n, k in ((64, 64), (63, 65)):
        _check(cco, [5, 30, 50, 60, -3], [15, 20, -4, 1000, 3], 90, n, k, torch.float32, 4)


@pytest.mark.parametrize("n,k", [(2048, 2048), (4096, 256), (512, 7168)])
def test_many_tiles_and_wide_tiles(cco, n, k):
    count = [300, 17, 513, 128, 129, 5, 700, 256]
    first = [sum(count[:i]) for i in range(len(count))]
    _check(cco, first, count, sum(count), n, k, torch.bfloat16, 5)


def test_small_tiles_for_a_short_last_round(cco):
    # 32 uneven groups of 256 rows on average: 320 tiles of 256 would be two
    # rounds of the 256 CUs, the second nearly empty
    g = torch.Generator().manual_seed(8)
    count = (256 + torch.randint(-60, 61, (32,), generator=g)).tolist()
    count[3] = 0
    count[-1] += 8192 - sum(count)
    first = [sum(count[:i]) for i in range(32)]
    for dtype in (torch.bfloat16, torch.float32):
        _check(cco, first, count, 8192, 2048, 144, dtype, 13)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", [(16, 256, 14336), (40, 512, 8192), (3, 128, 131056)])
def test_split_reductions(cco, dtype, rows, n, k):
    # few tiles and long sums: with workspace (the binding's) and without
    _check(cco, [0], [rows], rows, n, k, dtype, 6)
    from combine_symmetric_memory_amd import _capi
    import ctypes
    x, w = _codes((rows, k), 7).cuda(), _codes((1, n, k), 8).cuda()
    xs, ws = _scales(rows, 9).cuda(), _scales((1, n), 10, 1e-6).cuda()
    f, c = _i32([0]), _i32([rows])
    y = cco.group_product_i8(f, c, x, xs, w, ws, dtype=dtype)
    g = _capi.cco_groups(1, rows, f.data_ptr(), c.data_ptr())
    assert _capi.lib.cco_group_product_i8_workspace(ctypes.byref(g), n, k) > 0
    z = torch.empty_like(y)
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dtype]
    assert _capi.lib.cco_group_product_i8(
        ctypes.byref(g), x.data_ptr(), k, xs.data_ptr(), 1, w.data_ptr(), ws.data_ptr(), n, k,
        z.data_ptr(), code, n, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, z)  # integers: the same sums in any order


@pytest.mark.parametrize("n,k,ldx,ldy,shift", [(64, 64, 80, 72, 0), (64, 64, 64, 64, 16),
                                              (64, 64, 64, 64, 1), (64, 64, 65, 67, 0),
                                              (60, 96, 96, 64, 0), (72, 100, 112, 80, 3)])
def test_strides_and_alignments(cco, n, k, ldx, ldy, shift):
    for dtype in DTYPES:
        _check(cco, [0, 40], [40, 33], 75, n, k, dtype, 11, (ldx, ldy), 3, shift)


def test_the_largest_sums(cco):
    # |sum| up to 2^14 (2^17 - 1) stays inside an int32
    for k in (131071, 131056):
        x = torch.full((2, k), -128, dtype=torch.int8)
        x[1] = 127
        w = torch.full((1, 16, k), -128, dtype=torch.int8)
        one = torch.ones(2), torch.ones(1, 16)
        y = cco.group_product_i8(_i32([0]), _i32([2]), x.cuda(), one[0].cuda(), w.cuda(),
                                 one[1].cuda(), dtype=torch.float32)
        assert bool((y[0].double() == float(torch.tensor(16384.0 * k))).all())
        assert bool((y[1].double() == float(torch.tensor(-16256.0 * k))).all())


def test_scales_that_are_not_numbers_or_zero(cco):
    for n, k in ((64, 128), (65, 129)):
        x, w = _codes((40, k), 1), _codes((1, n, k), 2)
        xs, ws = _scales(40, 3), _scales((1, n), 4)
        xs[3], xs[5], ws[0, 9] = math.nan, 0.0, math.inf
        y = cco.group_product_i8(_i32([0]), _i32([40]), x.cuda(), xs.cuda(), w.cuda(), ws.cuda(),
                                 dtype=torch.float32).cpu()
        assert bool(torch.isnan(y[3]).all())
        keep = torch.arange(n) != 9
        assert not bool(y[5, keep].any())
        assert bool(torch.isfinite(y[[0, 1, 2, 4]][:, keep]).all())
        assert not bool(torch.isfinite(y[0, 9]))


def test_no_rows_and_no_groups_rows(cco):
    w, ws = _codes((2, 16, 32), 1).cuda(), _scales((2, 16), 2).cuda()
    y = cco.group_product_i8(_i32([0, 0]), _i32([0, 0]), torch.empty(0, 32, dtype=torch.int8,
                                                                     device="cuda"),
                             torch.empty(0, device="cuda"), w, ws)
    assert y.shape == (0, 16) and y.dtype == torch.bfloat16
    out = torch.full((4, 16), 3.0, device="cuda")
    cco.group_product_i8(_i32([0, 0]), _i32([0, 0]), _codes((4, 32), 3).cuda(),
                         torch.ones(4, device="cuda"), w, ws, out=out)
    assert bool((out == 3.0).all())


def test_many_groups(cco):
    G = 1024
    count = [(7 * g) % 3 for g in range(G)]
    first = [sum(count[:i]) for i in range(G)]
    _check(cco, first, count, sum(count), 32, 32, torch.float32, 12)


def test_repeats_streams_and_a_graph(cco):
    count = [300, 0, 17, 600]
    first = [0, 300, 300, 317]
    x, w = _codes((917, 1024), 1).cuda(), _codes((4, 768, 1024), 2).cuda()
    xs, ws = _scales(917, 3).cuda(), _scales((4, 768), 4).cuda()
    f, c = _i32(first), _i32(count)
    want = cco.group_product_i8(f, c, x, xs, w, ws)
    for _ in range(5):
        assert torch.equal(cco.group_product_i8(f, c, x, xs, w, ws), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cco.group_product_i8(f, c, x, xs, w, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    src = torch.randn(917, 1024, device="cuda").to(torch.bfloat16)
    with torch.cuda.stream(side):
        q, s = cco.quant_rows(src)
        cco.group_product_i8(f, c, q, s, w, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = cco.quant_rows(src)
        y = cco.group_product_i8(f, c, q, s, w, ws)
    for seed in range(3):
        src.copy_(torch.randn(917, 1024, generator=torch.Generator().manual_seed(seed)))
        eq, es = cco.quant_rows(src)
        ey = cco.group_product_i8(f, c, eq, es, w, ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, eq) and torch.equal(s, es) and torch.equal(y, ey)
