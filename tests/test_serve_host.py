"""Refusals of the 8-bit operators and of the layer for a few tokens, found on
the host before anything is launched (no GPU needed), and their binding's
checks."""
import ctypes

import pytest
import torch

P = 1 << 20  # a non-NULL, well aligned address that no refused call follows
META = torch.device("meta")


@pytest.fixture(scope="module")
def capi():
    from combine_symmetric_memory_amd import _capi
    return _capi


@pytest.fixture(scope="module")
def ops():
    from combine_symmetric_memory_amd import ops
    return ops


def test_quant_rows(capi):
    Q = capi.lib.cco_quant_rows
    big = 1 << 21
    #     x  dtype ldx rows cols swiglu q ldq s lds
    ok = [P, 0, 16, 4, 8, 1, P, 8, P, 1]
    for i, v in ((0, None), (0, P + 1), (1, 3), (1, -1), (2, 15), (2, big), (3, -1), (4, 0),
                 (4, -8), (4, 9), (6, None), (7, 7), (7, big), (8, None), (8, P + 2), (9, 0),
                 (9, -1), (9, 1 << 40)):
        a = list(ok)
        a[i] = v
        assert Q(*a, None) == -1, (i, v)
    assert Q(P + 2, 2, 16, 4, 8, 1, P, 8, P, 1, None) == -1  # fp32 at 2 bytes
    assert Q(P, 0, big, 4, big, 0, P, big, P, 1, None) == -1
    assert Q(None, 0, 16, 0, 8, 1, None, 8, None, 1, None) == 0


def _groups(capi, groups=4, rows=16, first=P, count=P):
    return ctypes.byref(capi.cco_groups(groups, rows, first, count))


def test_group_product_i8(capi):
    L, g = capi.lib.cco_group_product_i8, _groups(capi)
    big = 1 << 21
    #     x  ldx xs ldxs w ws n k y out ldy ws bytes
    ok = [P, 16, P, 1, P, P, 8, 16, P, 0, 8, None, 0]
    for i, v in ((0, None), (1, 15), (1, big), (2, None), (2, P + 2), (3, 0), (3, 1 << 40),
                 (4, None), (5, None), (5, P + 1), (6, 0), (6, big), (6, 9), (7, 0), (7, 17),
                 (8, None), (8, P + 1), (9, 3), (9, -1), (10, 7), (10, big)):
        a = list(ok)
        a[i] = v
        assert L(g, *a, None) == -1, (i, v)
    # the longest reduction whose sums fit
    assert L(g, P, 1 << 17, P, 1, P, P, 8, 1 << 17, P, 0, 8, None, 0, None) == -1
    for kw in (dict(groups=0), dict(groups=1025), dict(rows=-1), dict(first=None),
               dict(count=None), dict(first=P + 2)):
        assert L(_groups(capi, **kw), *ok, None) == -1
    assert L(None, *ok, None) == -1
    assert L(_groups(capi, rows=0), None, 16, None, 1, None, None, 8, 16, None, 0, 8, None, 0,
             None) == 0


def test_group_product_i8_workspace(capi):
    W, L = capi.lib.cco_group_product_i8_workspace, capi.lib.cco_group_product_i8
    one = _groups(capi, 1, 16)
    n = W(one, 256, 16384)
    assert n > 0 and n % (16 * 256 * 4) == 0
    for a in ((one, 256, 128), (one, 257, 16384), (one, 256, 16385), (one, 0, 16384),
              (one, 256, 1 << 17), (_groups(capi, 1, 0), 256, 16384), (None, 256, 16384)):
        assert W(*a) == 0
    for ws, size in ((P, n - 1), (P + 8, n)):
        assert L(one, P, 16384, P, 1, P, P, 256, 16384, P, 0, 256, ws, size, None) == -1


def _few(capi, H=64, I=32, E=4, K=2, dtype=0, wdtype=0, w13=P, w2=P, s13=None, s2=None):
    return ctypes.byref(capi.cco_few_desc(H, I, E, K, dtype, wdtype, w13, w2, s13, s2))


@pytest.mark.parametrize("kw", [dict(H=0), dict(I=0), dict(H=(1 << 20) + 1), dict(I=(1 << 19) + 1),
                                dict(E=0), dict(E=1025), dict(K=0), dict(K=33), dict(dtype=2),
                                dict(dtype=3, wdtype=3), dict(wdtype=1), dict(wdtype=2),
                                dict(dtype=-1, wdtype=-1)])
def test_few_shapes(capi, kw):
    d = _few(capi, **kw)
    assert capi.lib.cco_moe_few_workspace(d, 4) == 0
    assert capi.lib.cco_moe_few(d, P, P, P, 4, P, P, 1 << 40, None) == -1


def test_few_arguments(capi):
    F, W = capi.lib.cco_moe_few, capi.lib.cco_moe_few_workspace
    d = _few(capi)
    need = W(d, 4)
    assert need == 4 * 2 * 2 * 256 * 2  # T K rows of two planes of I, whole chunks
    ok = [P, P, P, 4, P, P, need]
    for i, v in ((0, None), (0, P + 1), (1, None), (1, P + 2), (2, None), (2, P + 2), (3, -1),
                 (4, None), (4, P + 1), (5, None), (5, P + 8), (6, need - 1)):
        a = list(ok)
        a[i] = v
        assert F(d, *a, None) == -1, (i, v)
    for kw in (dict(w13=None), dict(w2=None), dict(w13=P + 1), dict(w2=P + 1), dict(s13=P),
               dict(s2=P), dict(wdtype=3), dict(wdtype=3, s13=P), dict(wdtype=3, s2=P),
               dict(wdtype=3, s13=P + 2, s2=P)):
        assert F(_few(capi, **kw), *ok, None) == -1, kw
    assert F(None, *ok, None) == -1 and W(None, 4) == 0
    # too many tokens; none
    assert F(d, P, P, P, 65, P, P, 1 << 30, None) == -7 and W(d, 65) == 0 and W(d, -1) == 0
    assert F(d, None, None, None, 0, None, None, 0, None) == 0 and W(d, 0) == 0


def test_binding_refuses_host_tensors(ops):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(4, 8, dtype=torch.int8)
    w = torch.zeros(2, 8, 8, dtype=torch.int8)
    for call in (lambda: ops.quant_rows(x), lambda: ops.quant_swiglu(x),
                 lambda: ops.group_product_i8(i, i, q, torch.zeros(4), w, torch.zeros(2, 8)),
                 lambda: ops.moe_few(x, i.view(2, 1), torch.zeros(2, 1), w, w)):
        with pytest.raises(ValueError):
            call()


def test_scale_vectors(ops):
    def meta(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=META)

    assert ops._distance(meta(6), META, "s", 6) == 1
    assert ops._distance(meta(6, 5)[:, 2], META, "s", 6) == 5
    assert ops._distance(meta(1, 5)[:, 0], META, "s", 1) == 1
    for bad in (meta(5), meta(6, 1), meta(6, dtype=torch.float16), meta(1).expand(6), None,
                torch.zeros(6)):
        with pytest.raises(ValueError):
            ops._distance(bad, META, "s", 6)
