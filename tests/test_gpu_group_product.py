"""The products grouped by expert (cco_group_product and its gradients)
against 64-bit products: both kernels (rows of whole 16 bytes and any other),
ragged and empty groups, rows of no group, row distances, counts that reach
outside, accumulation, streams and graphs."""
import itertools

import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _rand(shape, dtype, seed, std=1.0, ld=None):
    """A tensor on the GPU, with row distance ld when given (the pad holds
    NaN: it must not be read into a result)."""
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(shape, generator=g) * std).to(dtype)
    if ld is None:
        return t.cuda()
    buf = torch.full((shape[0], ld), float("nan"), dtype=dtype)
    buf[:, :shape[1]] = t
    return buf.cuda()[:, :shape[1]]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _packed(counts):
    first = [0] + list(itertools.accumulate(counts))[:-1]
    return first, list(counts)


def _check_all(cco, first, count, rows, n, k, dtype, pads=(0, 0), seed=0, out_types=None):
    """The three products of one grouping; rows outside the groups keep what
    they held."""
    G = len(first)
    f, c = _i32(first), _i32(count)
    x = _rand((rows, k), dtype, seed, ld=k + pads[0] if pads[0] else None)
    dy = _rand((rows, n), dtype, seed + 1, ld=n + pads[1] if pads[1] else None)
    w = _rand((G, n, k), dtype, seed + 2, 0.1)
    parts = ref.rows_of(first, count, rows)
    xc, dc, wc = x.cpu(), dy.cpu(), w.cpu()
    for name, a, cols in (("product", x, n), ("dx", dy, k)):
        say("case: %s G=%d rows=%d n=%d k=%d %s pads=%s" % (name, G, rows, n, k, dtype, pads))
        pad = pads[1] if name == "product" else pads[0]
        buf = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
        out = buf[:, :cols]
        fn = cco.group_product if name == "product" else cco.group_product_dx
        fn(f, c, a, w, out=out)
        torch.cuda.synchronize()
        want = torch.full((rows, cols), 7.0, dtype=torch.float64)
        bound = torch.zeros((rows, cols), dtype=torch.float64)
        for g, (lo, hi) in enumerate(parts):
            if hi > lo:
                m = wc[g].t() if name == "product" else wc[g]
                v, s = ref.product((xc if name == "product" else dc)[lo:hi], m)
                want[lo:hi] = v
                bound[lo:hi] = ref.product_bound(v, s, m.shape[0], dtype)
        ref.assert_within(out, want, bound, name)
        if pad:
            assert bool((buf[:, cols:] == 7.0).all()), name + " wrote past its rows"
    for ot in out_types or (dtype, F32):
        say("case: dw G=%d rows=%d n=%d k=%d %s -> %s" % (G, rows, n, k, dtype, ot))
        out = torch.full((G, n, k), float("nan"), dtype=ot, device="cuda")
        cco.group_product_dw(f, c, dy, x, out=out)
        torch.cuda.synchronize()
        for g, (lo, hi) in enumerate(parts):
            v, s = ref.product(dc[lo:hi].t(), xc[lo:hi])
            ref.assert_within(out[g], v, ref.product_bound(v, s, hi - lo, ot), "dw group %d" % g)


SHAPES = [
    # counts, n, k
    ([1], 8, 8),
    ([1], 1, 1),
    ([5], 64, 64),
    ([0, 0, 3, 0], 16, 24),
    ([1, 2, 31, 32, 33, 0, 63, 64, 65], 96, 72),
    ([127, 128, 129], 256, 64),
    ([255, 256, 257, 1], 264, 136),
    ([300, 40, 700], 520, 328),
    ([130, 17], 512, 2048),
    ([20, 0, 9], 2048, 512),
    ([64] * 9, 1024, 256),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_packed_groups(cco, counts, n, k, dtype):
    first, count = _packed(counts)
    _check_all(cco, first, count, sum(counts), n, k, dtype, seed=n + k)


@pytest.mark.parametrize("counts,n,k", [([3, 50], 33, 65), ([140, 1, 0, 77], 129, 131),
                                        ([9], 257, 7), ([200], 7, 257), ([70, 300], 250, 190)])
def test_odd_sizes(cco, counts, n, k):
    first, count = _packed(counts)
    _check_all(cco, first, count, sum(counts), n, k, BF, seed=n * k)


@pytest.mark.parametrize("pads", [(8, 16), (1, 3), (64, 8), (5, 0)])
def test_row_distances(cco, pads):
    first, count = _packed([37, 0, 140, 64])
    _check_all(cco, first, count, 241, 136, 200, BF, pads=pads, seed=4)


def test_rows_of_no_group_and_any_order(cco):
    # gaps before, between and behind the groups, which are not in row order
    first, count = [300, 10, 0, 150, 399], [60, 100, 0, 33, 1]
    _check_all(cco, first, count, 410, 136, 72, BF, seed=9)
    _check_all(cco, first, count, 410, 33, 65, BF, seed=9)


def test_counts_that_reach_outside(cco):
    # rows below 0 and at or past `rows` are cut off; negative counts are none
    first, count = [-5, 20, 90, 200, 50], [15, 30, 1000, 7, -3]
    _check_all(cco, first, count, 100, 64, 48, BF, seed=3)
    first, count = [2 ** 31 - 8, -2 ** 31, 0], [100, 2 ** 31 - 1, 2 ** 31 - 1]
    _check_all(cco, first, count, 40, 64, 48, BF, seed=3, out_types=(F32,))


def test_shared_rows_in_the_weight_gradient(cco):
    first, count = [0, 10, 0], [40, 30, 0]
    x, dy = _rand((60, 72), BF, 1), _rand((60, 40), BF, 2)
    dw = cco.group_product_dw(_i32(first), _i32(count), dy, x)
    for g in range(3):
        lo, hi = first[g], first[g] + count[g]
        v, s = ref.product(dy[lo:hi].cpu().t(), x[lo:hi].cpu())
        ref.assert_within(dw[g], v, ref.product_bound(v, s, hi - lo, BF), "group %d" % g)


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("n,k", [(136, 264), (33, 65)])
def test_accumulate(cco, ot, n, k):
    first, count = _packed([50, 0, 200])
    x, dy = _rand((250, k), BF, 1), _rand((250, n), BF, 2)
    old = _rand((3, n, k), ot, 3)
    out = old.clone()
    cco.group_product_dw(_i32(first), _i32(count), dy, x, out=out, accumulate=True)
    for g in range(3):
        lo, hi = first[g], first[g] + count[g]
        v, s = ref.product(dy[lo:hi].cpu().t(), x[lo:hi].cpu())
        o = old[g].cpu().double()
        b = ref.product_bound(v + o, s + o.abs(), hi - lo + 1, ot)
        ref.assert_within(out[g], v + o, b, "group %d" % g)
    # without rows nothing changes
    zero = _i32([0, 0, 0])
    keep = out.clone()
    cco.group_product_dw(zero, zero, dy, x, out=out, accumulate=True)
    assert torch.equal(out, keep)
    cco.group_product_dw(zero, zero, dy[:0], x[:0], out=out, accumulate=True)
    assert torch.equal(out, keep)
    cco.group_product_dw(zero, zero, dy[:0], x[:0], out=out)
    assert not out.any()


def test_infinities_stay_in_their_rows(cco):
    # a bad row of one group, a bad pad and a bad weight of another group
    # reach nothing else
    first, count = _packed([70, 5, 90])
    x = _rand((165, 72), BF, 1, ld=80)
    w = _rand((3, 136, 72), BF, 2)
    x[72] = float("inf")
    x[3, 5] = float("nan")
    w[1, 7] = float("nan")
    y = cco.group_product(_i32(first), _i32(count), x, w).float().cpu()
    bad = torch.zeros(165, 136, dtype=torch.bool)
    bad[3] = True
    bad[72] = True
    bad[70:75, 7] = True
    assert torch.isfinite(y[~bad]).all()
    assert (~torch.isfinite(y[3])).all() and torch.isnan(y[70:75, 7]).all()
    # the reduction of dw ends with the group's rows
    dy = _rand((165, 136), BF, 3)
    dw = cco.group_product_dw(_i32(first), _i32(count), dy, x).float().cpu()
    assert torch.isfinite(dw[2]).all() and not torch.isfinite(dw[1]).any()
    dx = cco.group_product_dx(_i32(first), _i32(count), dy, w).float().cpu()
    assert torch.isnan(dx[70:75]).all() and torch.isfinite(dx[:70]).all() \
        and torch.isfinite(dx[75:]).all()


def test_many_groups(cco):
    counts = [(i * 7919) % 5 for i in range(1024)]
    first, count = _packed(counts)
    _check_all(cco, first, count, sum(counts), 24, 40, BF, seed=6, out_types=(BF,))


def test_the_same_bits_every_time_and_other_streams(cco):
    first, count = _packed([100, 0, 333, 47])
    f, c = _i32(first), _i32(count)
    x, dy, w = _rand((480, 520), BF, 1), _rand((480, 264), BF, 2), _rand((4, 264, 520), BF, 3)
    base = (cco.group_product(f, c, x, w), cco.group_product_dx(f, c, dy, w),
            cco.group_product_dw(f, c, dy, x))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i in range(4):  # two streams at once
        s = s1 if i % 2 else s2
        got.append((cco.group_product(f, c, x, w, stream=s),
                    cco.group_product_dx(f, c, dy, w, stream=s),
                    cco.group_product_dw(f, c, dy, x, stream=s)))
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, base):
            assert torch.equal(a, b)


def test_captured_into_a_graph_with_changing_groups(cco):
    x, dy, w = _rand((300, 264), BF, 1), _rand((300, 136), BF, 2), _rand((3, 136, 264), BF, 3)
    f, c = _i32([0, 100, 200]), _i32([100, 100, 100])
    y = torch.zeros((300, 136), dtype=BF, device="cuda")
    dx = torch.zeros((300, 264), dtype=BF, device="cuda")
    dw = torch.zeros((3, 136, 264), dtype=F32, device="cuda")

    def run():
        cco.group_product(f, c, x, w, out=y)
        cco.group_product_dx(f, c, dy, w, out=dx)
        cco.group_product_dw(f, c, dy, x, out=dw)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for counts in ([100, 100, 100], [300, 0, 0], [1, 2, 250], [0, 0, 0]):
        first, count = _packed(counts)
        f.copy_(_i32(first))
        c.copy_(_i32(count))
        for t in (y, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.zero_()
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(cco):
    # rows past 2^31 elements of the row operand: the last group's rows lie
    # behind 4 GiB
    rows, k, n = 300_000, 7168, 64
    x = torch.zeros((rows, k), dtype=BF, device="cuda")
    tail = _rand((40, k), BF, 1)
    x[-40:] = tail
    w = _rand((2, n, k), BF, 2)
    f, c = _i32([0, rows - 40]), _i32([3, 40])
    y = cco.group_product(f, c, x, w)
    v, s = ref.product(tail.cpu(), w[1].cpu().t())
    ref.assert_within(y[-40:], v, ref.product_bound(v, s, k, BF), "rows behind 4 GiB")
    dy = torch.zeros((rows, n), dtype=BF, device="cuda")
    dy[-40:] = _rand((40, n), BF, 3)
    dw = cco.group_product_dw(f, c, dy, x)
    v, s = ref.product(dy[-40:].cpu().t(), tail.cpu())
    ref.assert_within(dw[1], v, ref.product_bound(v, s, 40, BF), "dw behind 4 GiB")
    dx = x  # overwritten row by row
    cco.group_product_dx(f, c, dy, w, out=dx)
    v, s = ref.product(dy[-40:].cpu(), w[1].cpu())
    ref.assert_within(dx[-40:], v, ref.product_bound(v, s, n, BF), "dx behind 4 GiB")


@pytest.mark.parametrize("counts,n,k", [([40], 128, 2048), ([3, 0, 17], 72, 4104),
                                        ([1], 2056, 64), ([2100], 64, 72), ([9000, 0, 5], 40, 136)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_split_reductions(cco, counts, n, k, dtype):
    # few tiles and long reductions in one of the three directions
    first, count = _packed(counts)
    _check_all(cco, first, count, sum(counts), n, k, dtype, pads=(8, 8), seed=n)


def test_a_split_reduction_needs_its_workspace_and_keeps_other_rows(cco):
    import ctypes
    from combine_symmetric_memory_amd import _capi
    n, k, rows = 136, 4096, 90
    x, w = _rand((rows, k), BF, 1), _rand((2, n, k), BF, 2)
    f, c = _i32([70, 0]), _i32([15, 50])
    g = _capi.cco_groups(2, rows, f.data_ptr(), c.data_ptr())
    nbytes = _capi.lib.cco_group_product_workspace(0, ctypes.byref(g), n, k)
    assert nbytes > 0
    ws = torch.full((nbytes + 64,), 7, dtype=torch.uint8, device="cuda")
    outs = []
    for p, size in ((None, 0), (ws.data_ptr(), nbytes)):
        out = torch.full((rows, n), 3.0, dtype=BF, device="cuda")
        assert _capi.lib.cco_group_product(ctypes.byref(g), 0, x.data_ptr(), k, w.data_ptr(), n, k,
                                           out.data_ptr(), n, p, size,
                                           torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert bool((out[50:70] == 3).all()) and bool((out[85:] == 3).all())
        for lo, hi, e in ((70, 85, 0), (0, 50, 1)):
            v, s = ref.product(x[lo:hi].cpu(), w[e].cpu().t())
            ref.assert_within(out[lo:hi], v, ref.product_bound(v, s, k, BF), "group %d" % e)
        outs.append(out)
    assert bool((ws[nbytes:] == 7).all())


def test_smallest_numbers(cco):
    # subnormal operands, products and results count like any others
    f, c = _i32([0]), _i32([33])
    for dtype, tiny in ((HF, 2.0 ** -22), (BF, 2.0 ** -130)):
        g = torch.Generator().manual_seed(1)
        x = (torch.randint(-3, 4, (33, 72), generator=g) * tiny).to(dtype)
        w = torch.randint(-2, 3, (1, 40, 72), generator=g).to(dtype)
        for k in (72, 65):
            y = cco.group_product(f, c, x[:, :k].contiguous().cuda(),
                                  w[:, :, :k].contiguous().cuda())
            want = x[:, :k].double() @ w[0, :, :k].double().t()
            # sums of few integers times tiny: exact before the one rounding
            bound = ref.half_step(dtype) * want.abs() + ref.smallest(dtype)
            ref.assert_within(y, want, bound, "%s k=%d" % (dtype, k))


@pytest.mark.parametrize("rows,n,k,groups", [(80, 64, 7168, 2), (4096, 64, 512, 1),
                                             (300, 264, 520, 3), (2000, 2048, 2048, 7),
                                             (40, 4096, 128, 2)])
def test_repeats_are_equal_bit_for_bit(cco, rows, n, k, groups):
    # every tile form, split and not, into poisoned outputs: a store that
    # takes a register too late shows as a few wrong elements now and then
    counts = [rows // groups] * groups
    first, count = _packed(counts)
    f, c = _i32(first), _i32(count)
    rows = sum(counts)
    x, dy, w = _rand((rows, k), BF, 1), _rand((rows, n), BF, 2), _rand((groups, n, k), BF, 3)
    old = _rand((groups, n, k), F32, 4)
    outs = [torch.empty((rows, n), dtype=BF, device="cuda"),
            torch.empty((rows, k), dtype=BF, device="cuda"),
            torch.empty((groups, n, k), dtype=BF, device="cuda"),
            torch.empty((groups, n, k), dtype=F32, device="cuda"),
            torch.empty((groups, n, k), dtype=F32, device="cuda"),
            torch.empty((groups, n, k), dtype=BF, device="cuda")]

    def run():
        for o in outs[:4]:
            o.fill_(float("nan"))
        outs[4].copy_(old)
        outs[5].copy_(old)
        cco.group_product(f, c, x, w, out=outs[0])
        cco.group_product_dx(f, c, dy, w, out=outs[1])
        cco.group_product_dw(f, c, dy, x, out=outs[2])
        cco.group_product_dw(f, c, dy, x, out=outs[3])
        cco.group_product_dw(f, c, dy, x, out=outs[4], accumulate=True)
        cco.group_product_dw(f, c, dy, x, out=outs[5], accumulate=True)

    run()
    want = [o.clone() for o in outs]
    assert torch.allclose(want[3] + old, want[4], atol=1e-4, rtol=1e-5)
    assert bool((want[3].to(BF) == want[2]).all())
    differ = torch.zeros(len(outs), dtype=torch.int64, device="cuda")
    for _ in range(50):
        run()
        for i, o in enumerate(outs):
            differ[i] += (o != want[i]).sum()
    assert differ.tolist() == [0] * len(outs)


@pytest.mark.parametrize("per,groups,n,k", [(30, 70, 2048, 2048), (3, 1000, 4096, 136),
                                            (300, 1000, 1024, 128), (290, 900, 136, 1288)])
def test_more_tiles_than_workgroups(cco, per, groups, n, k):
    # workgroups take several tiles, full and wide ones in turn: a tile's
    # first loads and the last tile's stores are in flight together
    g = torch.Generator().manual_seed(per)
    counts = (torch.randint(0, 2 * per + 1, (groups,), generator=g)).tolist()
    first, count = _packed(counts)
    rows = sum(counts)
    f, c = _i32(first), _i32(count)
    gen = torch.Generator(device="cuda").manual_seed(7)

    def r(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(BF)

    x, dy, w = r(rows, k), r(rows, n), r(groups, n, k)
    outs = [torch.empty((rows, n), dtype=BF, device="cuda"),
            torch.empty((rows, k), dtype=BF, device="cuda"),
            torch.empty((groups, n, k), dtype=BF, device="cuda"),
            torch.empty((groups, n, k), dtype=F32, device="cuda")]

    def run():
        for o in outs:
            o.fill_(float("nan"))
        cco.group_product(f, c, x, w, out=outs[0])
        cco.group_product_dx(f, c, dy, w, out=outs[1])
        cco.group_product_dw(f, c, dy, x, out=outs[2])
        cco.group_product_dw(f, c, dy, x, out=outs[3])

    run()
    want = [o.clone() for o in outs]
    for e in (0, 1, groups // 2, groups - 2, groups - 1):
        lo, hi = first[e], first[e] + count[e]
        xs, ds, we = x[lo:hi].cpu(), dy[lo:hi].cpu(), w[e].cpu()
        for i, (a, b, terms) in enumerate(((xs, we.t(), k), (ds, we, n), (ds.t(), xs, hi - lo),
                                           (ds.t(), xs, hi - lo))):
            v, s = ref.product(a, b)
            got = want[i][lo:hi] if i < 2 else want[i][e]
            ref.assert_within(got, v, ref.product_bound(v, s, terms, outs[i].dtype),
                              "output %d group %d" % (i, e))
    assert bool((want[3].to(BF) == want[2]).all())
    differ = torch.zeros(4, dtype=torch.int64, device="cuda")
    for _ in range(15):
        run()
        for i, o in enumerate(outs):
            differ[i] += (o != want[i]).sum()
    assert differ.tolist() == [0] * 4
