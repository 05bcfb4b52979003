"""The 8-bit operators and the layer for a few tokens where offsets pass 32
bits: rows and weights behind the first 4 GiB, against the same call on those
alone."""
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_rows_past_4_gib(cco):
    # 5.4 GB of rows, 2.7 GB of codes
    rows, cols = 82000, 32768
    x = torch.zeros(rows, cols, dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-7:] = torch.randn(7, cols, generator=g, device="cuda").half()
    q, s = cco.quant_rows(x)
    want, ws = cco.quant_rows(x[-7:].clone())
    assert torch.equal(q[-7:], want) and torch.equal(s[-7:], ws)
    assert not bool(q[:-7].any()) and not bool(s[:-7].any())


@pytest.mark.parametrize("k", [8192, 8200])
def test_weights_past_4_gib(cco, k):
    # the fast kernel and, with rows of 8-byte alignment, the general one
    G, n, rows = 66, 8192, 300
    say("case: i8 weights past 4 GiB, k=%d" % k)
    w = torch.zeros(G, n, k, dtype=torch.int8, device="cuda")
    assert w.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(2)
    w[-1] = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(rows, device="cuda"), torch.rand(G, n, device="cuda")
    first, count = [0] * G, [0] * G
    count[-1] = rows
    y = cco.group_product_i8(_i32(first), _i32(count), x, xs, w, ws, dtype=torch.float32)
    one = cco.group_product_i8(_i32([0]), _i32([rows]), x, xs, w[-1:].clone(), ws[-1:].clone(),
                               dtype=torch.float32)
    assert bool(y.any()) and torch.equal(y, one)


def test_results_past_4_gib(cco):
    # 4.4 GB of results; rows and their results at the far end
    rows, n, k = 68000, 16384, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (1, n, k), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(rows, device="cuda"), torch.rand(1, n, device="cuda")
    y = cco.group_product_i8(_i32([0]), _i32([rows]), x, xs, w, ws, dtype=torch.float32)
    far = slice(rows - 40, rows)
    one = cco.group_product_i8(_i32([0]), _i32([40]), x[far].clone(), xs[far].clone(), w, ws,
                               dtype=torch.float32)
    assert torch.equal(y[far], one)


@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("T", [2, 40])
def test_experts_past_4_gib(cco, wdtype, T):
    # the last expert's weights lie behind 4 GiB of both matrices
    i8 = wdtype == torch.int8
    E, H, I = (70, 4096, 16384) if i8 else (70, 4096, 8192)
    say("case: few past 4 GiB %s T=%d" % (wdtype, T))
    g = torch.Generator(device="cuda").manual_seed(4)

    def last(shape):
        if i8:
            return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        return (torch.randn(shape, generator=g, device="cuda") * 0.02).to(wdtype)

    w13 = torch.zeros(E, 2 * I, H, dtype=wdtype, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=wdtype, device="cuda")
    w13[-1], w2[-1] = last((2 * I, H)), last((H, I))
    s13 = torch.full((E, 2 * I), 2e-4, device="cuda") if i8 else None
    s2 = torch.full((E, H), 2e-4, device="cuda") if i8 else None
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
    w = torch.rand(T, 1, generator=g, device="cuda")
    y = cco.moe_few(x, idx, w, w13, w2, s13=s13, s2=s2)
    # (70 experts and one may take different forms, whose sums differ in order)
    xf = x.double()
    a, b = w13[-1].double(), w2[-1].double()
    if i8:
        a, b = a * 2e-4, b * 2e-4
    gu = xf @ a.t().contiguous()
    h = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
    want = (h @ b.t().contiguous()) * w.double()
    bound = 2.0 ** -8 * want.abs() + 1e-4 * float(want.abs().max())
    assert bool(((y.double() - want).abs() <= bound).all())
