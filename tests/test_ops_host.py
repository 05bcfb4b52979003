"""Refusals of the operators in include/cco_ops.h, found on the host before
anything is launched (no GPU needed), and their binding's checks."""
import ctypes

import pytest
import torch

P = 1 << 20  # a non-NULL, well aligned address that no refused call follows


@pytest.fixture(scope="module")
def capi():
    from combine_symmetric_memory_amd import _capi
    return _capi


def _route(capi, E=8, K=2, score=0, renorm=0, scale=1.0, groups=1, kept=1):
    return ctypes.byref(capi.cco_route_desc(E, K, score, renorm, scale, groups, kept))


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=1025), dict(K=0), dict(K=33, E=64), dict(K=9),
                                dict(score=2), dict(groups=0), dict(groups=3), dict(groups=65),
                                dict(groups=4, kept=5), dict(groups=4, kept=0),
                                dict(groups=4, kept=1, K=3)])
def test_route_shapes(capi, kw):
    d = _route(capi, **kw)
    assert capi.lib.cco_route(d, P, 2, 1 << 20, None, 4, P, P, None) == -1


@pytest.mark.parametrize("args", [(None, 2, 8, None, 4, P, P), (P, 3, 8, None, 4, P, P),
                                  (P, 2, 7, None, 4, P, P), (P, 2, 8, P + 2, 4, P, P),
                                  (P, 2, 8, None, -1, P, P), (P, 2, 8, None, 4, None, P),
                                  (P, 2, 8, None, 4, P, None), (P + 2, 2, 8, None, 4, P, P),
                                  (P + 1, 0, 8, None, 4, P, P), (P, 2, 8, None, 4, P + 1, P),
                                  (P, 2, 8, None, 4, P, P + 2)])
def test_route_arguments(capi, args):
    assert capi.lib.cco_route(_route(capi), *args, None) == -1


def test_route_without_tokens_and_descriptor(capi):
    assert capi.lib.cco_route(_route(capi), None, 2, 8, None, 0, None, None, None) == 0
    assert capi.lib.cco_route(None, P, 2, 8, None, 4, P, P, None) == -1
    L = capi.lib.cco_route_grad
    assert L(_route(capi), None, 2, 8, None, None, 0, None, 8, None) == 0
    for a in ((None, 2, 8, P, P, 4, P, 8), (P, 2, 8, None, P, 4, P, 8), (P, 2, 8, P, None, 4, P, 8),
              (P, 2, 8, P, P, 4, None, 8), (P, 2, 8, P, P, 4, P, 7), (P, 2, 7, P, P, 4, P, 8),
              (P, 5, 8, P, P, 4, P, 8), (P, 2, 8, P + 2, P, 4, P, 8), (P, 2, 8, P, P, 4, P + 1, 8)):
        assert L(_route(capi), *a, None) == -1


def _groups(capi, groups=4, rows=16, first=P, count=P):
    return ctypes.byref(capi.cco_groups(groups, rows, first, count))


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=1025), dict(rows=-1),
                                dict(first=None), dict(count=None), dict(first=P + 2)])
def test_groups(capi, kw):
    g = _groups(capi, **kw)
    L = capi.lib
    assert L.cco_group_product(g, 0, P, 8, P, 8, 8, P, 8, None, 0, None) == -1
    assert L.cco_group_product_dx(g, 0, P, 8, P, 8, 8, P, 8, None, 0, None) == -1
    assert L.cco_group_product_dw(g, 0, P, 8, P, 8, 8, 8, P, 0, 0, None, 0, None) == -1


def test_group_product_arguments(capi):
    L, g = capi.lib, _groups(capi)
    big = 1 << 22
    for a in ((2, P, 8, P, 8, 8, P, 8), (0, None, 8, P, 8, 8, P, 8), (0, P, 7, P, 8, 8, P, 8),
              (0, P, 8, None, 8, 8, P, 8), (0, P, 8, P, 0, 8, P, 8), (0, P, 8, P, 8, 0, P, 8),
              (0, P, 8, P, 8, 8, None, 8), (0, P, 8, P, 8, 8, P, 7), (0, P + 1, 8, P, 8, 8, P, 8),
              (0, P, 8, P + 1, 8, 8, P, 8), (0, P, 8, P, 8, 8, P + 1, 8), (9, P, 8, P, 8, 8, P, 8),
              (0, P, big, P, 8, 8, P, 8), (0, P, 8, P, big, 8, P, big)):
        assert L.cco_group_product(g, *a, None, 0, None) == -1, a
        assert L.cco_group_product_dx(g, *a, None, 0, None) == -1, a
    for a in ((2, P, 8, P, 8, 8, 8, P, 2, 0), (0, P, 8, P, 8, 8, 8, P, 1, 0),
              (0, P, 7, P, 8, 8, 8, P, 0, 0), (0, P, 8, P, 7, 8, 8, P, 0, 0),
              (0, P, 8, P, 8, 8, 8, None, 0, 0), (0, P, 8, P, 8, 8, 8, P + 2, 2, 0),
              (0, None, 8, P, 8, 8, 8, P, 0, 0)):
        assert L.cco_group_product_dw(g, *a, None, 0, None) == -1, a
    assert L.cco_group_product(None, 0, P, 8, P, 8, 8, P, 8, None, 0, None) == -1
    # no rows: nothing to do, and nothing launched
    none = _groups(capi, rows=0)
    assert L.cco_group_product(none, 0, None, 8, P, 8, 8, None, 8, None, 0, None) == 0
    assert L.cco_group_product_dx(none, 0, None, 8, P, 8, 8, None, 8, None, 0, None) == 0
    assert L.cco_group_product_dw(none, 0, None, 8, None, 8, 8, 8, P, 0, 1, None, 0, None) == 0


def test_group_workspace(capi):
    L = capi.lib
    W = L.cco_group_product_workspace
    # few tiles and a long reduction: parts of the fp32 result
    one = _groups(capi, groups=1, rows=64)
    n = W(capi.CCO_GROUP_PRODUCT, one, 256, 8192)
    assert n > 0 and n % (64 * 256 * 4) == 0 and n // (64 * 256 * 4) >= 2
    assert W(capi.CCO_GROUP_DX, one, 8192, 256) > 0
    assert W(capi.CCO_GROUP_DW, _groups(capi, groups=1, rows=8192), 64, 256) > 0
    # none where nothing is split: many tiles, short reductions, rows of
    # other than whole 16 bytes, no rows, bad arguments
    assert W(capi.CCO_GROUP_PRODUCT, _groups(capi, groups=64, rows=65536), 4096, 8192) == 0
    assert W(capi.CCO_GROUP_PRODUCT, one, 256, 64) == 0
    assert W(capi.CCO_GROUP_PRODUCT, one, 257, 8192) == 0
    assert W(capi.CCO_GROUP_PRODUCT, _groups(capi, rows=0), 256, 8192) == 0
    assert W(3, one, 256, 8192) == 0 and W(0, None, 256, 8192) == 0
    # too small or misaligned
    for ws, size in ((P, n - 1), (P + 8, n)):
        assert L.cco_group_product(one, 0, P, 8192, P, 256, 8192, P, 256, ws, size, None) == -1


def _norm(capi, H=64, dtype=0, wdtype=2, kind=0, eps=1e-6, post=None, gate=None, pre=P):
    return capi.cco_block_norm_desc(H, dtype, wdtype, kind, 1.0, eps, post, gate, pre)


@pytest.mark.parametrize("kw", [dict(H=0), dict(H=16385), dict(dtype=3), dict(wdtype=1),
                                dict(kind=3, gate=P), dict(kind=0, gate=P), dict(kind=1),
                                dict(kind=2), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(pre=P + 2), dict(post=P + 2), dict(kind=2, gate=P + 2),
                                dict(dtype=0, wdtype=0, pre=P + 1)])
def test_norm_descriptors(capi, kw):
    d = ctypes.byref(_norm(capi, **kw))
    L = capi.lib
    assert L.cco_block_norm(d, P, P, 4, P, P, None) == -1
    assert L.cco_block_norm_grad_workspace(d, 4) == 0
    assert L.cco_block_norm_grad(d, P, P, P, P, 4, P, P, None, None, P, P, 1 << 30, None) == -1


def test_norm_arguments(capi):
    L, d = capi.lib, ctypes.byref(_norm(capi))
    for a in ((None, P, 4, P, P), (P, P, -1, P, P), (P, P, 4, P, None), (P, None, 4, P, P),
              (P, P, 4, None, None), (P + 1, P, 4, P, P), (P, P + 1, 4, P, P),
              (P, P, 4, P + 1, P), (P, P, 4, P, P + 1)):
        assert L.cco_block_norm(d, *a, None) == -1, a
    nopre = ctypes.byref(_norm(capi, pre=None))
    assert L.cco_block_norm(nopre, P, P, 4, P, P, None) == -1   # u without pre
    assert L.cco_block_norm(nopre, P, None, 4, None, None, None) == -1
    assert L.cco_block_norm(ctypes.byref(_norm(capi, post=P)), P, None, 4, None, P, None) == -1
    assert L.cco_block_norm(d, None, None, 0, None, None, None) == 0
    ws = L.cco_block_norm_grad_workspace(d, 4)
    assert ws == 4 * 64 * 4
    G = L.cco_block_norm_grad
    ok = [P, P, P, P, 4, P, P, None, None, P, P, ws]
    for i, v in ((0, None), (1, None), (3, None), (4, -1), (5, None), (6, None), (7, P), (8, P),
                 (9, None), (10, None), (10, P + 8), (11, ws - 1), (0, P + 1), (9, P + 2)):
        a = list(ok)
        a[i] = v
        assert G(d, *a, None) == -1, (i, v)
    # neither gradient
    assert G(nopre, P, P, None, None, 4, P, P, None, None, None, P, ws, None) == -1
    M = L.cco_moe_combine_norm
    assert M(None, P, d, P, 4, None, P, P, None) == -1


def test_binding_refuses_host_tensors_and_shapes(capi):
    import combine_symmetric_memory_amd as cco
    x = torch.zeros(4, 8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        cco.route(x, 2)
    with pytest.raises(ValueError):
        cco.route_grad(x, i, x)
    with pytest.raises(ValueError):
        cco.group_product(i, i, x.bfloat16(), torch.zeros(2, 8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        cco.group_product_dw(i, i, x.bfloat16(), x.bfloat16())
    with pytest.raises(ValueError):
        cco.block_norm(x, x, pre=torch.ones(8))
    with pytest.raises(ValueError):
        cco.block_norm_grad(x, x, x)
